// Large-M kernel instances, fp16, with adapters.
#define W4A16_BF 0
#define W4A16_LORA
#include "w4a16_large.inc"
