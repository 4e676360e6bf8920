// The experts' large products, fp16.
#define W4A16_BF 0
#include "w4a16_experts_large.inc"
