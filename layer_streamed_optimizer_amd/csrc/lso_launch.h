// Kernel launches that report their own error.
#pragma once

#include <hip/hip_runtime.h>

namespace lso {

template <typename T>
struct as_is {
    typedef T type;
};

// Launch kernel(args...) and return the launch's own error.  hipGetLastError
// would also give, and take away, what other code of this thread left there;
// only an error of this launch, which the caller gets, is taken from it.
template <typename... P>
hipError_t launch(void (*kernel)(P...), dim3 grid, dim3 threads, hipStream_t s, const typename as_is<P>::type&... args)
{
    void* list[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    const hipError_t err = hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, threads, list, 0, s);
    if (err != hipSuccess) (void)hipGetLastError();
    return err;
}

}  // namespace lso
