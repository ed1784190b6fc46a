// Host check of the norm and rotation's arguments: of a side without heads no
// pointer or stride reaches the kernel, whatever the caller left there; and of
// its split: the parts of all tokens fit on the card together, and one more of
// each would not, unless a token has no more passes.
#include <cstdio>
#include <cstring>

#include "tq_q8.cuh"

int main() {
  int bad = 0;
  for (int hq : {0, 3})
    for (int hk : {0, 3}) {
      tq_qk_norm_rope_args x;
      std::memset(&x, 0, sizeof(x));
      x.batch = 1, x.n = 2, x.num_q_heads = hq, x.num_kv_heads = hk, x.head_dim = 128, x.eps = 1e-6f;
      x.q = (void*)16, x.k = (void*)32, x.q_weight = (void*)49, x.k_weight = (void*)65, x.q_out = (void*)80, x.k_out = (void*)96;
      x.q_row_stride = 8, x.q_token_stride = 16, x.q_head_stride = 24, x.k_row_stride = 32, x.k_token_stride = 40, x.k_head_stride = 48;
      x.positions = (int32_t*)128, x.inv_freq = (float*)144, x.interleaved = 1;
      const tq::NormRopeArgs a = tq::norm_rope_args(x);
      bad += a.q != (hq ? x.q : nullptr) || a.q_weight != (hq ? x.q_weight : nullptr) || a.q_out != (hq ? x.q_out : nullptr);
      bad += a.k != (hk ? x.k : nullptr) || a.k_weight != (hk ? x.k_weight : nullptr) || a.k_out != (hk ? x.k_out : nullptr);
      bad += a.q_row != (hq ? 8 : 0) || a.q_token != (hq ? 16 : 0) || a.q_head != (hq ? 24 : 0);
      bad += a.k_row != (hk ? 32 : 0) || a.k_token != (hk ? 40 : 0) || a.k_head != (hk ? 48 : 0);
      bad += a.batch != 1 || a.n != 2 || a.Hq != hq || a.Hkv != hk || a.d != 128 || a.eps != 1e-6f || a.interleaved != 1 ||
             a.positions != x.positions || a.inv_freq != x.inv_freq;
    }
  for (int warps : {20, 2960, 3000})
    for (int passes : {1, 2, 3, 10, 16})
      for (int64_t tokens : {1, 2, 8, 19, 20, 21, 185, 296, 700, 1000, 1479, 1480, 1481, 1776, 2960, 2961, 12297, 2147483647}) {
        const int64_t parts = tq::norm_rope_parts(tokens, passes, warps);
        bad += parts < 1 || parts > passes || (parts > 1 && tokens * parts > warps) ||
               (parts < passes && tokens * (parts + 1) <= warps);
      }
  std::printf(bad ? "bad %d\n" : "ok\n", bad);
  return bad != 0;
}
