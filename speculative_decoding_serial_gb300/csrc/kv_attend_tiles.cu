// kv_attend_tiles.cu — attention of many rows without first keys that stay visible.
#include "kv_attend_tiles.cuh"

namespace whead_kv_impl {
template int launch_tiles<false>(const HostCache& h, const AttendArgs& a, int max_q);
}
