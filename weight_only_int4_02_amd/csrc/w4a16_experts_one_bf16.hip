// The experts' products for one token, bfloat16.
#define W4A16_BF 1
#include "w4a16_experts_one.inc"
