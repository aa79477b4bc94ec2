// The WKV7 operators of libwkv7.so, one translation unit: the sticky device status
// word (status.cuh) is one __device__ variable shared by their kernels, so they are
// compiled together (no relocatable device code needed).  The state-space mixer's
// files, which have no such word, are units of their own.
#include "wkv7_api.cu"
#include "fwd_seq.cu"
#include "step.cu"
#include "bwd_chunk.cu"
#include "bwd_chunk_tc.cu"
#include "bwd_dchain.cu"
#include "fwd_chunk.cu"
#include "bwd_noalloc.cu"
#include "fwd_host.cu"
#include "timemix.cu"
