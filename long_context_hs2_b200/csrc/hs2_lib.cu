// libhs2's translation unit: the hybrid block's entry points and the paged decode
// path's, which use the former's host helpers.
#include "hs2_api.cu"

#include "paged_api.cuh"
