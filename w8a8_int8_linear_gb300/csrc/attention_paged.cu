// Attention of new tokens over a cache in pages.
#include "attention.cuh"

namespace w8a8 {

size_t paged_attention_workspace_bytes(int num_sms) { return attention_workspace_bytes(num_sms); }

cudaError_t launch_paged_attention(const AttentionArgs& args, int max_queries, int dtype, int num_sms, void* workspace,
                                   void* encode_fn, cudaStream_t st, char* detail, size_t n) {
    AttentionArgs a = args;
    a.few_rows = 0;
    a.most_rows = 0x7FFFFFFF;
    a.expected_rows = max_queries * a.group;
    return launch_attention_split(a, dtype, num_sms, workspace, encode_fn, st, detail, n);
}

}  // namespace w8a8
