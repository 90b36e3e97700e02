// Attention over a paged cache of int8 codes, head dimension 128: a file for each, so that they compile side by side.
#define LFM2SC_CACHED8_D 128
#define LFM2SC_CACHED8_INT8 true
#include "attn_cached8.hpp"
