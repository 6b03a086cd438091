// The prompts' kernels with weights of 8 bits (attn_prefill.cuh), how a call is split, and
// the way to either set of kernels.
#include "attn_prefill.cuh"

namespace fp8moe {

void plan_prefill(PrefillArgs *a, int d, int sms, const PrefillFit &fit) {
  // pieces of at most 16 heads, as even as may be
  const int per_kv = a->n_heads / a->n_kv;
  a->chunks = (per_kv + 15) / 16;
  a->heads = (per_kv + a->chunks - 1) / a->chunks;
  a->tokens = 128 / a->heads;
  const int T = a->tokens * (d == 256 ? 1 : 2);
  a->items = ((int64_t)a->Tq / T + a->B) * a->n_kv * a->chunks;
  // Few items leave SMs idle: a cluster then shares an item's blocks, where all clusters are
  // resident at once and the blocks that a CTA is spared take longer than the join.  By the
  // sequences' mean lengths, which are what the host knows; times in ns, of two full
  // tiles.  us without and with (d 128 unless told):
  //   1 query, 8001 keys, 32/8 heads        88   20.8 (8)
  //   64 queries, 2064 keys, 32/8           32.7 22.4 (4)
  //   128 queries, 8128 keys, 32/8          103  40.1 (4)
  //   128 queries, 4128 keys, 16/8, d 256   62.2 28.8 (4)
  //   1000 queries, 5000 keys, 16/1         66.0 48.2 (2)
  //   1 query, 501 keys, 16/16              11.4 10.0 (4)
  //   500 queries and keys, 16/16           13.5 15.5 (4), 18.4 (2): not taken
  a->splits = 1;
  const int keys = d == 256 ? 64 : 128;
  const int64_t mean_q = ((int64_t)a->Tq + a->B - 1) / a->B, tokens = mean_q < T ? mean_q : T;
  int64_t blocks = ((int64_t)a->Tk / a->B + keys - 1) / keys;
  if (a->window > 0 && (a->window + tokens) / keys + 2 < blocks) blocks = (a->window + tokens) / keys + 2;
  const int64_t block_ns = d == 256 ? 900 : 1500, join_ns = 2000 + 8000 * tokens / T;
  int64_t best = blocks * block_ns;
  for (int i = 0; i < kSplitSizes; ++i) {
    const int splits = 2 << i;
    const int64_t resident = fit.clusters[i] < sms / splits ? fit.clusters[i] : sms / splits;
    const int64_t ns = (blocks + splits - 1) / splits * block_ns + join_ns;
    if (a->items <= resident && ns < best) best = ns, a->splits = splits;
  }
}

cudaError_t ready_prefill16(int d, PrefillFit *fit);
cudaError_t launch_prefill16(const PrefillArgs &a, int d, int sms, cudaStream_t s);

cudaError_t ready_prefill(int d, int bits, PrefillFit *fit) { return bits == 16 ? ready_prefill16(d, fit) : ready_terms<1>(d, fit); }

cudaError_t launch_prefill(const PrefillArgs &a, int d, int bits, int sms, cudaStream_t s) {
  return bits == 16 ? launch_prefill16(a, d, sms, s) : launch_terms<1>(a, d, sms, s);
}

}  // namespace fp8moe
