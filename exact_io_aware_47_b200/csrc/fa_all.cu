// Single translation unit of the library: the device status word is shared
// by every kernel without relocatable device code.
#include "fa_api.cu"
#include "fa_fwd.cu"
#include "fa_bwd.cu"
#include "fa_quant.cu"
#include "fa_rope.cu"
#include "fa_cache.cu"
#include "fa_tree.cu"
#include "fa_serve_api.cu"
