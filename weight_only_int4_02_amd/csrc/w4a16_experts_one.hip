// The experts' products for one token, fp16.
#define W4A16_BF 0
#include "w4a16_experts_one.inc"
