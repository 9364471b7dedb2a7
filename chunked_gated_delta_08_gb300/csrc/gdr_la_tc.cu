// gdr_la_tc.cu -- linear attention on the tcgen05 tensor cores (not built yet: every pass takes gdr_la.cu's form).
#include "gdr_la.cuh"

namespace gdr {
namespace la {

bool tc_takes(const LaArgs &, int, int) { return false; }
int launch_tc(const LaArgs &, int, cudaStream_t) { return GDR_ERR_UNSUPPORTED; }

}  // namespace la
}  // namespace gdr
