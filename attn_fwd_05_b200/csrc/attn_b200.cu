// attn_b200.cu — the library's one translation unit: the attention entry points and the 4-bit
// cache and page entry points of include/attn_b200.h.  They share the device status word and
// the host helpers of attn_api.cu.
#include "attn_api.cu"
#include "cache_api.cuh"
