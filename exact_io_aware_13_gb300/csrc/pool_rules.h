// How many CTAs the clusters of the pool's plans and of the verification have: plain functions of
// sizes, without CUDA, so that tests run them on the host.
#pragma once

namespace attn {

constexpr int kPlanMaxCtas = 16;   // the largest cluster there is
constexpr int kPortableCtas = 8;   // the largest that every device of this kind schedules
constexpr int kVerifyCtasPerSm = 4;
constexpr int kVerifyEach = 4096;  // tokens of a CTA, a step of its warps' vector loads or two

// CTAs of a plan: one up to `one` units of work, else one per `each`, as a power of two.
constexpr int plan_ctas(long long work, int one, int each) {
  int n = 1;
  while (work > one && n < kPlanMaxCtas && (long long)n * each < work) n *= 2;
  return n;
}

// CTAs per sequence of a verification: what the SMs hold at once, shared by the sequences, and a step
// of the warps' vector loads each at least. Clusters of sixteen only for up to a 24th of the CTAs that
// the SMs hold (25 sequences: they do not pack as closely as small ones, and do not all start at once)
// and from sixteen steps on; nothing between eight and sixteen. Microseconds by eight and by sixteen:
// 256000 fp32 tokens 13.0 and 9.1 for 4 sequences, 18.7 and 13.5 for 24, 22.7 and 24.8 for 38; 100000
// bf16 tokens 7.6 and 6.9, 8.9 and 9.7, 10.0 and 14.0; 50257 bf16 tokens 6.6 and 6.4, 7.6 and 8.9, 8.2 and
// 12.8 (by thirteen 6.4 for 4 sequences, 8.9 for 38); 64 sequences over 256000 bf16 tokens 21.4 by eight,
// 26.2 by nine.
constexpr int verify_ctas(int num_sms, int B, int V) {
  const long long held = (long long)num_sms * kVerifyCtasPerSm / B, steps = (long long)V / kVerifyEach + 1;
  const long long ctas = steps < held ? steps : held > 1 ? held : 1;
  if (ctas <= kPortableCtas) return (int)ctas;
  return steps >= kPlanMaxCtas && held >= 24 ? kPlanMaxCtas : kPortableCtas;
}

}  // namespace attn
