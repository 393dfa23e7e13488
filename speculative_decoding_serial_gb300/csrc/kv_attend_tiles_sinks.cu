// kv_attend_tiles_sinks.cu — attention of many rows with a window and first keys that stay visible behind it. 2 x 2048 tokens, window
// 1,024, 100 first keys: 145 us as without those (75 GFLOP, 0.52 PFLOP/s): an item has ten blocks, and the change from one to the next, some 12
// us, and the blocks that masks cut (13 us in all) weigh more than in long items.
#include "kv_attend_tiles.cuh"

namespace whead_kv_impl {
template int launch_tiles<true>(const HostCache& h, const AttendArgs& a, int max_q);
}
