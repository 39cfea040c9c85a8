// linear_backward.hip - the products dz w and dz^T x of linear_act_backward, in tiles.

#include "linear_products.h"

namespace mgg_dense {
template mgg_status run_product<false, false, true, false>(const Product&, TileArgs, hipStream_t);
template mgg_status run_product<false, true, true, false>(const Product&, TileArgs, hipStream_t);
template mgg_status run_product<true, false, true, false>(const Product&, TileArgs, hipStream_t);
template mgg_status run_product<true, true, true, false>(const Product&, TileArgs, hipStream_t);
}  // namespace mgg_dense
