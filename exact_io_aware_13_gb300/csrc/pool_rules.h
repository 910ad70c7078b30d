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
// of the warps' vector loads each at least; nothing between eight and sixteen. Clusters of sixteen do
// not fill the SMs: 33 of them start at once, so they are left to 32 sequences (19 CTAs held for each),
// and to rows of sixteen steps. Microseconds by sixteen and by eight: 32 sequences over 256000 fp32 tokens
// 15.1 and 20.9, 34 of them 21.6 and 22.0, of bf16 12.6 and 13.4, then 15.6 and 13.8; over 100000 bf16 tokens
// 4 sequences 6.9 and 7.6, 32 9.9 and 9.0, 34 12.9 and 8.9; over 50257 bf16 tokens 4 sequences 6.4 and 6.6, 24 8.9
// and 7.6, 38 12.8 and 8.2 (by thirteen 6.4, -, 8.9). 64 sequences over 256000 bf16 tokens 21.4 by eight, 26.2
// by nine.
constexpr int verify_ctas(int num_sms, int B, int V) {
  const long long held = (long long)num_sms * kVerifyCtasPerSm / B, steps = (long long)V / kVerifyEach + 1;
  const long long ctas = steps < held ? steps : held > 1 ? held : 1;
  if (ctas <= kPortableCtas) return (int)ctas;
  return steps >= kPlanMaxCtas && held >= 19 ? kPlanMaxCtas : kPortableCtas;
}

}  // namespace attn
