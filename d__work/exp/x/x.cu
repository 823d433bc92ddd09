#include "pgd_prefill.cuh"
template __global__ void pgd::prefill_kernel<128,false>(const __grid_constant__ pgd::PrefillMaps, const pgd::PrefillParams);
