// What the chunk kernels take a sequence to be, for tests on the CPU: the
// function that the kernels call, over host memory.
#include "attn_chunk.cuh"

extern "C" void chunk_sequence(int packed, const int32_t* starts, const int32_t* table, const int32_t* lens,
                               int64_t n_seqs, int64_t T, int64_t max_pages, int page_size, int64_t b, int* out) {
    gbe::ChunkArgs a = {};
    a.packed = packed != 0;
    a.starts = starts, a.table = table, a.lens = lens;
    a.n_seqs = n_seqs, a.T = T, a.max_pages = max_pages, a.c.page_size = page_size;
    const gbe::chunk::Seq s = gbe::chunk::sequence(a, b);
    out[0] = s.begin, out[1] = s.n, out[2] = s.len;
}
