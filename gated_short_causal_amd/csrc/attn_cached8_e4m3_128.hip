// Attention over a paged cache of e4m3 codes, head dimension 128: a file for each, so that they compile side by side.
#define LFM2SC_CACHED8_D 128
#define LFM2SC_CACHED8_INT8 false
#include "attn_cached8.hpp"
