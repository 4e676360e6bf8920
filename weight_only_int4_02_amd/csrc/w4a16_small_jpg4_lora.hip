// Small-M kernel instances for 4 MFMA step(s) per group, fp16, with adapters.
#define W4A16_JPG 4
#define W4A16_BF 0
#define W4A16_LORA
#include "w4a16_small_inst.inc"
