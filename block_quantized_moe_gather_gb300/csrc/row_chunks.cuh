// How rows are cut into chunks, for any int number of rows.  Plain arithmetic,
// so that it compiles for the host alone too (the tests do that).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define BQ_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define BQ_HOST_DEVICE inline
#endif

namespace bq {

// Chunks of at most `most` rows that `rows` >= 0 rows make.
BQ_HOST_DEVICE int row_chunks(int rows, int most) {
    return (int)(((uint32_t)rows + (uint32_t)most - 1u) / (uint32_t)most);
}

struct RowChunk {
    int first, rows;
};

// Chunk i of `chunks` of near-equal size that `rows` >= 1 rows are cut into.
// With chunks = row_chunks(rows, most), size <= most and (chunks - 1) * most <
// rows: every chunk has a row, and i * size stays below `rows`.
BQ_HOST_DEVICE RowChunk row_chunk(int rows, int chunks, int i) {
    const int size = (rows - 1) / chunks + 1, first = i * size;
    return {first, size < rows - first ? size : rows - first};
}

// a + b, or limit + 1 where the sum is more than `limit` (0 <= a, b <= limit + 1,
// limit < 2^30).  Sums of chunks that pass the limit stay there instead of
// wrapping, in whatever order they are added.
BQ_HOST_DEVICE int add_chunks(int a, int b, int limit) {
    const uint32_t sum = (uint32_t)a + (uint32_t)b;
    return sum > (uint32_t)limit ? limit + 1 : (int)sum;
}

}  // namespace bq
