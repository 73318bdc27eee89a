// The library's one translation unit: the square attention entry points
// (fa_lib.cu), and the entry points for keys of another length, caches, spans of
// keys, caches in pages, and the head norm and rotation, which use the same checks,
// launch helpers and device status word.
#include "fa_lib.cu"

#include "fa_cross.cuh"
#include "fa_cross_fwd.cuh"
#include "fa_cross_bwd.cuh"
#include "fa_span.cuh"
#include "fa_span_fwd.cuh"
#include "fa_span_few.cuh"
#include "fa_span_bwd.cuh"
#include "fa_rope.cuh"
#include "fa_cross_api.cuh"
#include "fa_span_api.cuh"
#include "fa_rope_api.cuh"
