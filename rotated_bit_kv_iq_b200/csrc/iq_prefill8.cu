// Causal attention of a chunk of query tokens over the 8-bit cache: the two kernels that it may take.
#include <algorithm>

#include "iq_prefill8_tc.cuh"

namespace iq {

size_t prefill8_workspace_bytes(int batch, int n_tok, int n_q_heads, int n_kv_heads, int max_ctx) {
  const int g = std::min(8, n_q_heads / n_kv_heads);
  return std::max(pt_plan(batch, n_tok, g, n_kv_heads, max_ctx).bytes, chunk8_workspace_bytes(batch, n_tok, g, n_kv_heads));
}

// 16-bit queries on tcgen05; float32 queries, whose outputs are to be right to 2^-20 or so, with two binary16 terms of q
// and of P on mma.sync (decode8_kernel).
int launch_prefill8(const View8& v, const void* q, int dtype, int batch, int n_tok, int n_q_heads, const int32_t* start,
                    const int32_t* n_valid, int max_ctx, float scale, void* out, void* workspace, void* stream) {
  if (batch == 0 || n_tok == 0) return 0;
  if (dtype == IQ_F32)
    return launch_chunk8(v, q, dtype, batch, n_tok, n_q_heads, start, n_valid, max_ctx, scale, out, workspace, stream);
  return launch_prefill8_tc(v, q, dtype, batch, n_tok, n_q_heads, start, n_valid, max_ctx, scale, out, workspace, stream);
}

}  // namespace iq
