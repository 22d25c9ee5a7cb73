// The causal convolution's kernels for every element type and width.
#include "conv.cuh"
#include "sequence.h"

namespace selinv {
namespace {

// Calls f with the width as a compile-time number.
template <class F> cudaError_t with_width(int k, F f)
{
    switch (k) {
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    case 8: return f(std::integral_constant<int, 8>());
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

template <class T> cudaError_t conv_launch(const ConvArgs &p, cudaStream_t s)
{
    return with_width(p.k, [&](auto k) { return conv_run<T, k.value>(p, s); });
}
template <class T> cudaError_t conv_backward_launch(const ConvArgs &p, cudaStream_t s)
{
    return with_width(p.k, [&](auto k) { return conv_backward_run<T, k.value>(p, s); });
}
template <class T> cudaError_t conv_step_launch(const ConvStepArgs &p, cudaStream_t s)
{
    return with_width(p.k, [&](auto k) { return conv_step_run<T, k.value>(p, s); });
}

#define SELINV_CONV_INSTANCES(T)                                              \
    template cudaError_t conv_launch<T>(const ConvArgs &, cudaStream_t);      \
    template cudaError_t conv_backward_launch<T>(const ConvArgs &, cudaStream_t); \
    template cudaError_t conv_step_launch<T>(const ConvStepArgs &, cudaStream_t);
SELINV_CONV_INSTANCES(double)
SELINV_CONV_INSTANCES(float)
SELINV_CONV_INSTANCES(__nv_bfloat16)
SELINV_CONV_INSTANCES(__half)

}  // namespace selinv
