// Internal launcher declarations of the softmax-attention layer's kernels: the
// q/k norm with the rotation, the paged key/value cache and the tree attention
// over it. Arguments are validated by the C-ABI layer (attn_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Multiprocessors of the current device (148 where there is none).
int sm_count();

// Address of the device status word on the current device (api.cu).
int* device_status_ptr();

// Paged cache: k, v [n_pages, Hk, page, D], scales [n_pages, Hk, page] (e4m3).
struct CacheView {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t n_pages;
    int page_shift;  // page = 1 << page_shift tokens
    int Hk, D;
    int e4m3;  // 1: e4m3 values with fp32 scales, 0: bf16 values
};

// Where the packed tokens stand: sequence n's tokens cu[n]..cu[n+1] are the
// last of its lens[n] cached positions; position p is row p % page of page
// table[n * max_pages + p / page].
struct PageArgs {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu;
    int N, max_pages;
};

struct RowsArgs {
    const void* q;  // [T, H, D], token stride ld_q (elements)
    const void* k;  // [T, Hk, D]
    const void* v;  // [T, Hk, D] (cache modes)
    int64_t ld_q, ld_k, ld_v;
    int is_bf16;
    int64_t T;
    int H, Hk, D;
    const float* q_w;
    const float* k_w;
    float eps;
    const int32_t* pos;      // [T]
    const double* inv_freq;  // [rotary / 2]
    int rotary, interleaved;
    void* q_out;  // [T, H, D] dense
    void* k_out;  // [T, Hk, D] dense (no cache)
    CacheView c;
    PageArgs p;
    int* status;
};
enum RowsMode : int { kNormRope = 0, kNormRopeCache = 1, kCacheWrite = 2 };
cudaError_t launch_rows(const RowsArgs& a, RowsMode mode, cudaStream_t s);

struct ReadArgs {
    CacheView c;
    PageArgs p;
    int64_t T;
    void* k;  // [T, Hk, D] dense
    void* v;
    int out_bf16;
    int* status;
};
cudaError_t launch_kv_read(const ReadArgs& a, cudaStream_t s);

constexpr int kMaxNodes = 64;  // drafted tokens of one sequence (a node's mask is one 64-bit word)

struct AcceptArgs {
    CacheView c;
    PageArgs p;
    const int32_t* path;  // [N, M]
    int M;
    int32_t* new_lens;  // [N]
    int* status;
};
cudaError_t launch_kv_accept(const AcceptArgs& a, cudaStream_t s);

struct TreeArgs {
    const void* q;  // [T, H, D] bf16, token stride ld_q
    int64_t ld_q;
    CacheView c;
    PageArgs p;
    int64_t T;
    int H;
    const int64_t* mask;  // [T] or null: a chain
    int max_nodes;
    float scale;
    const void* gate;  // [T, H, D] bf16 or null
    void* o;           // [T, H, D] bf16 dense
    float* lse;        // [T, H] or null
    void* workspace;
    int* status;
    uint64_t wait_ns;  // bound on each wait of the tcgen05 kernel
    // the launch's plan (launch_tree_attention)
    int grid, row_tiles, slot_rows;
};
size_t tree_workspace_bytes(int N, int H, int Hk, int D, int max_nodes, int e4m3);
// The tcgen05 kernel alone, for a planned launch.
cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t s);
cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s);

}  // namespace gdn
