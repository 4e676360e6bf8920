// Small-M kernel instances for 2 MFMA step(s) per group, bfloat16, with adapters.
#define W4A16_JPG 2
#define W4A16_BF 1
#define W4A16_LORA
#include "w4a16_small_inst.inc"
