// int8_scales.cuh -- a sum of 8-bit integers' products times the scales of its token and channel.
//
// Token first, then channel.  A sum is an integer below 2^45, so with a scale of any size the
// product keeps 24 bits, and with one up to 2^80 it stays in fp32's range.  A larger token's
// scale comes last: the product before it leaves the range only where the result does.
#pragma once

namespace bwgemm {

__device__ __forceinline__ bool large_scale(float token)
{
    return fabsf(token) > 0x1p80f;
}

__device__ __forceinline__ float scaled_sum(float sum, float token, float channel)
{
    return large_scale(token) ? sum * channel * token : sum * token * channel;
}

}  // namespace bwgemm
