// lib.hip — the translation unit of libmoe.so: the block-quantized path
// (libmoe.hip), then the scored routing and the 8-bit float path, which share
// its error word, routing buffers and argument checks.
#include "libmoe.hip"

#include "fp8_quant.hip"
#include "route_scored.hip"
#include "fp8_skinny.hip"
#include "fp8_gemm.hip"
#include "fp8_api.hip"
