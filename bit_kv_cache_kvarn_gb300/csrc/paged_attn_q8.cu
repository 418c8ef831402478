// The kernels of paged_attn.cu over 8-bit caches, compiled beside those over 16-bit ones.
#define KVARN_PAGED_Q8 1
#include "paged_attn.cu"
