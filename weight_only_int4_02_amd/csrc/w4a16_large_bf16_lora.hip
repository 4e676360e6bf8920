// Large-M kernel instances, bfloat16, with adapters.
#define W4A16_BF 1
#define W4A16_LORA
#include "w4a16_large.inc"
