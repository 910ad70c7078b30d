// The cluster sizes of the pool's plans and of the verification, for the host's tests.
#include "pool_rules.h"

extern "C" {
int host_verify_ctas(int num_sms, int B, int V) { return attn::verify_ctas(num_sms, B, V); }
int host_plan_ctas(long long work, int one, int each) { return attn::plan_ctas(work, one, each); }
}
